// gdr_conv.cu -- short causal convolution per channel: forward, backward, and
// the single-token step with states in a pool of slots.
//
//   p_t = bias + sum_j w_j x_{t - W + 1 + j};  y_t = act(p_t)
//   backward, g_t = dy_t act'(p_t):  dx_t = sum_i w_{W-1-i} g_{t+i},  dw_j = sum_t g_t x_{t-W+1+j}
// with x_{-1}, .. x_{-W+1} taken from the sequence's state, and the last W - 1
// inputs of each sequence left as its new state.
//
// A thread owns VEC neighbouring channels and walks a run of tokens with the
// W - 1 inputs before in registers, so every input is read from HBM once (the
// W - 1 tokens around a run come from L2 again).  Runs are cut from the flat
// token axis; a sequence's border inside one reloads the window.  The bound is
// HBM.
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

template <typename T, int VEC, int W>
struct Taps {
  float w[W][VEC], bias[VEC];
  __device__ __forceinline__ void load(const ConvArgs &a, int64_t e) {
    const bool f32 = a.d.weight_dtype == GDR_F32;
    float v[W][VEC];  // the VEC * W weights are one run of memory
#pragma unroll
    for (int k = 0; k < W; ++k) {
      if (f32) load_vec<VEC>(static_cast<const float *>(a.weight) + e * W + k * VEC, v[k]);
      else load_vec<VEC>(static_cast<const T *>(a.weight) + e * W + k * VEC, v[k]);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][i] = v[(i * W + j) / VEC][(i * W + j) % VEC];
      bias[i] = a.bias ? param<T>(a.bias, f32, e + i) : 0.f;
    }
  }
};

// The W - 1 inputs before token t of sequence s (x rows, or rows of the state).
template <typename T, int VEC, int W>
__device__ __forceinline__ void load_window(const ConvArgs &a, const Seq &s, int64_t t, int64_t e,
                                            float (&win)[W][VEC]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int64_t u = t - (W - 1) + j;
    if (u >= s.bos) {
      load_vec<VEC>(static_cast<const T *>(a.x) + u * a.d.ld_x + e, win[j]);
    } else if (a.s0) {
      load_vec<VEC>(static_cast<const T *>(a.s0) + (s.n * (W - 1) + (u - s.bos + W - 1)) * a.d.E + e, win[j]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) win[j][i] = 0.f;
    }
  }
}

// States of sequences without tokens: `to` = `from` (zero where null).
template <typename T, int VEC, int W>
__device__ __forceinline__ void copy_empty(const ConvArgs &a, int64_t e, const void *from, void *to) {
  if (!to) return;
  for (int64_t n = 0; n < a.d.N; ++n) {
    const SeqRange r = seq_range(a.cu, n, a.d.T);
    if (r.eos > r.bos) continue;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      float v[VEC] = {};
      const int64_t at = (n * (W - 1) + j) * a.d.E + e;
      if (from) load_vec<VEC>(static_cast<const T *>(from) + at, v);
      store_vec<VEC>(static_cast<T *>(to) + at, v);
    }
  }
}

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvArgs a) {
  if (!seqlens_ok(a.cu, a.d.N, a.M, a.status)) return;
  const int64_t e = (int64_t)((blockIdx.x % a.tiles) * a.cx + threadIdx.x % a.cx) * VEC;
  const int64_t run = (int64_t)(blockIdx.x / a.tiles) * (kThreads / a.cx) + threadIdx.x / a.cx;
  if (e >= a.d.E) return;
  if (run == 0) copy_empty<T, VEC, W>(a, e, a.s0, a.st);
  int64_t t = run * a.L;
  const int64_t end = t + a.L < a.M ? t + a.L : a.M;
  if (t >= end) return;
  const bool silu = a.d.activation == GDR_ACT_SILU;
  Taps<T, VEC, W> p;
  p.load(a, e);
  Seq s = seq_at(a, t);
  float win[W][VEC];
  load_window<T, VEC, W>(a, s, t, e, win);
  const T *x = static_cast<const T *>(a.x) + e;
  T *y = static_cast<T *>(a.y) + e;
  constexpr int U = 4;  // tokens whose loads are in flight together
  for (; t < end; t += U) {
    float in[U][VEC];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t + u < end) load_vec<VEC>(x + (t + u) * a.d.ld_x, in[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t + u < end) {
        if (t + u == s.eos) {  // the next sequence that has tokens starts here
          s = seq_at(a, t + u);
          load_window<T, VEC, W>(a, s, t + u, e, win);
        }
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          win[W - 1][i] = in[u][i];
          o[i] = p.bias[i];
#pragma unroll
          for (int j = 0; j < W; ++j) o[i] = fmaf(p.w[j][i], win[j][i], o[i]);
          if (silu) o[i] *= sigmoid_fast(o[i]);
        }
        store_vec<VEC>(y + (t + u) * a.d.E, o);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
          for (int i = 0; i < VEC; ++i) win[j][i] = win[j + 1][i];
        if (a.st && t + u + 1 == s.eos) {
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
            store_vec<VEC>(static_cast<T *>(a.st) + (s.n * (W - 1) + j) * a.d.E + e, win[j]);
        }
      }
    }
  }
}

// Backward.  A run is taken sequence by sequence; for its tokens [ta, tb) the
// walk goes W - 1 further, because dx_t needs g up to token t + W - 1 (zero past
// the sequence).  At step u the gradient of token u - W + 1 is complete; where
// that is before the sequence it is the gradient of a row of the state.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(ConvArgs a) {
  if (!seqlens_ok(a.cu, a.d.N, a.M, a.status)) return;
  const int64_t e = (int64_t)((blockIdx.x % a.tiles) * a.cx + threadIdx.x % a.cx) * VEC;
  const int64_t run = (int64_t)(blockIdx.x / a.tiles) * (kThreads / a.cx) + threadIdx.x / a.cx;
  if (e >= a.d.E || run >= a.runs) return;
  if (run == 0) copy_empty<T, VEC, W>(a, e, a.dst, a.st);
  const int64_t t0 = run * a.L, end = t0 + a.L < a.M ? t0 + a.L : a.M;
  const bool silu = a.d.activation == GDR_ACT_SILU;
  Taps<T, VEC, W> p;
  p.load(a, e);
  float dw[W][VEC], db[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    db[i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
  }
  const T *x = static_cast<const T *>(a.x) + e, *dy = static_cast<const T *>(a.dy) + e;
  const T *dst = a.dst ? static_cast<const T *>(a.dst) + e : nullptr;
  T *dx = static_cast<T *>(a.y) + e, *ds0 = a.st ? static_cast<T *>(a.st) + e : nullptr;
  for (int64_t ta = t0; ta < end;) {
    const Seq s = seq_at(a, ta);
    const int64_t tb = s.eos < end ? s.eos : end;
    float win[W][VEC], g[W][VEC];
    load_window<T, VEC, W>(a, s, ta, e, win);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) g[j][i] = 0.f;
    constexpr int U = 4;
    const int64_t last = tb + W - 1;  // one past the last step
    for (int64_t t = ta; t < last; t += U) {
      float in[U][VEC], up[U][VEC];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t + u < last && t + u < s.eos) {
          load_vec<VEC>(x + (t + u) * a.d.ld_x, in[u]);
          load_vec<VEC>(dy + (t + u) * a.d.ld_dy, up[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t q = t + u;
        if (q >= last) continue;
        if (q < s.eos) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            win[W - 1][i] = in[u][i];
            float v = p.bias[i];
#pragma unroll
            for (int j = 0; j < W; ++j) v = fmaf(p.w[j][i], win[j][i], v);
            float gr = up[u][i];
            if (silu) {
              const float sg = sigmoid_fast(v);
              gr *= sg * fmaf(v, 1.f - sg, 1.f);
            }
            g[W - 1][i] = gr;
            if (q < tb) {
              db[i] += gr;
#pragma unroll
              for (int j = 0; j < W; ++j) dw[j][i] = fmaf(gr, win[j][i], dw[j][i]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) g[W - 1][i] = 0.f;
        }
        const int64_t to = q - (W - 1);  // complete now
        if (to >= ta || (ta == s.bos && ds0)) {
          float o[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            o[i] = 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) o[i] = fmaf(p.w[W - 1 - j][i], g[j][i], o[i]);
          }
          const int64_t row = to - s.eos + (W - 1);  // its row in the new state, if it is there
          if (dst && row >= 0) {
            float v[VEC];
            load_vec<VEC>(dst + (s.n * (W - 1) + row) * a.d.E, v);
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] += v[i];
          }
          if (to >= ta) store_vec<VEC>(dx + to * a.d.E, o);
          else store_vec<VEC>(ds0 + (s.n * (W - 1) + (to - s.bos + W - 1)) * a.d.E, o);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            win[j][i] = win[j + 1][i];
            g[j][i] = g[j + 1][i];
          }
      }
    }
    ta = tb;
  }
  float *part = a.part + run * (W + 1) * a.d.E + e;
#pragma unroll
  for (int j = 0; j < W; ++j) store_vec<VEC>(part + j * a.d.E, dw[j]);
  store_vec<VEC>(part + W * a.d.E, db);
}

// dweight [E, W] and dbias [E] from the runs' partials, added in run order.
__global__ void __launch_bounds__(256) conv_sum_kernel(const float *__restrict__ part, int64_t runs, int64_t E, int W,
                                                       float *__restrict__ dweight, float *__restrict__ dbias,
                                                       SeqCheck seqs) {
  __shared__ float sm[8][32];
  if (!seqlens_ok(seqs)) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, j = blockIdx.y;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float acc = 0.f;
  if (c < E) {
#pragma unroll 8
    for (int64_t r = w; r < runs; r += 8) acc += part[(r * (W + 1) + j) * E + c];
  }
  sm[w][lane] = acc;
  __syncthreads();
  if (w == 0 && c < E) {
#pragma unroll
    for (int i = 1; i < 8; ++i) acc += sm[i][lane];
    if (j < W) dweight[c * W + j] = acc;
    else if (dbias) dbias[c] = acc;
  }
}

// One token per row: window from the slot, shifted back with the new input.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvArgs a) {
  const int64_t e = (int64_t)((blockIdx.x % a.tiles) * a.cx + threadIdx.x % a.cx) * VEC;
  const int64_t r = (int64_t)(blockIdx.x / a.tiles) * (kThreads / a.cx) + threadIdx.x / a.cx;
  if (e >= a.d.E || r >= a.d.B) return;
  int64_t slot = a.slots ? a.slots[r] : r;
  if (slot >= a.d.N) {
    raise_status(a.status, GDR_ERR_SLOTS);
    slot = -1;
  }
  T *y = static_cast<T *>(a.y) + r * a.d.E + e;
  float o[VEC];
  if (slot < 0) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) o[i] = 0.f;
    store_vec<VEC>(y, o);
    return;
  }
  T *st = static_cast<T *>(a.st) + slot * (W - 1) * a.d.E + e;
  float win[W][VEC];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load_vec<VEC>(st + j * a.d.E, win[j]);
  load_vec<VEC>(static_cast<const T *>(a.x) + r * a.d.ld_x + e, win[W - 1]);
  Taps<T, VEC, W> p;
  p.load(a, e);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_vec<VEC>(st + j * a.d.E, win[j + 1]);
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    o[i] = p.bias[i];
#pragma unroll
    for (int j = 0; j < W; ++j) o[i] = fmaf(p.w[j][i], win[j][i], o[i]);
    if (a.d.activation == GDR_ACT_SILU) o[i] *= sigmoid_fast(o[i]);
  }
  store_vec<VEC>(y, o);
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

// Tokens in a run: long enough that the W - 1 tokens read again, the weights
// and (backward) the partials are small beside it, short enough that the grid
// fills the GPU.
int run_length(int64_t M, int64_t E, int vec, int lo, int hi) {
  const int64_t want = M * cdiv(E, vec) / ((int64_t)kSMs * 1024);
  int L = lo;
  while (L < hi && L < want) L *= 2;
  return L;
}

// Channels of a thread: VF in the forward and the step, VB in the backward.
template <typename T, int VF, int VB>
int launch(ConvArgs a, Dir dir, float *dweight, float *dbias, cudaStream_t st) {
  const gdr_conv_desc &d = a.d;
  const int VEC = dir == kBwd ? VB : VF;
  a.cx = channel_threads(d.E, VEC);
  const int64_t tiles = cdiv(d.E, (int64_t)VEC * a.cx), per = kThreads / a.cx;
  a.tiles = (unsigned)tiles;
  if (dir == kStep) {
    const int64_t blocks = tiles * cdiv(d.B, per);
    if (blocks > 0x7fffffff) return set_error(GDR_ERR_SHAPE, "too many rows for one launch");
    return with_taps(d.W, [&](auto w) {
      conv_step_kernel<T, VF, decltype(w)::value><<<(unsigned)blocks, kThreads, 0, st>>>(a);
      return launched("conv_step_kernel");
    });
  }
  a.L = dir == kFwd ? run_length(a.M, d.E, VEC, 8, 32) : run_length(a.M, d.E, VEC, 16, 128);
  a.runs = std::max<int64_t>(1, cdiv(a.M, a.L));
  const int64_t blocks = tiles * cdiv(a.runs, per);
  if (blocks > 0x7fffffff) return set_error(GDR_ERR_SHAPE, "too many tokens for one launch");
  if (dir == kFwd) {
    return with_taps(d.W, [&](auto w) {
      conv_fwd_kernel<T, VF, decltype(w)::value><<<(unsigned)blocks, kThreads, 0, st>>>(a);
      return launched("conv_fwd_kernel");
    });
  }
  char *base = nullptr;
  int rc = scratch_begin(sizeof(float) * (size_t)(a.runs * (d.W + 1) * d.E), st, "convolution backward scratch", &base);
  if (rc != GDR_OK) return rc;
  a.part = (float *)base;
  rc = with_taps(d.W, [&](auto w) {
    conv_bwd_kernel<T, VB, decltype(w)::value><<<(unsigned)blocks, kThreads, 0, st>>>(a);
    return launched("conv_bwd_kernel");
  });
  if (rc == GDR_OK) {
    conv_sum_kernel<<<dim3((unsigned)cdiv(d.E, 32), (unsigned)(d.W + (dbias ? 1 : 0))), 256, 0, st>>>(
        a.part, a.runs, d.E, (int)d.W, dweight, dbias, SeqCheck{a.cu, d.N, a.M, a.status});
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
  const int64_t E = a.d.E;
  const bool vec = E % 8 == 0 && a.d.ld_x % 8 == 0 && a.d.ld_dy % 8 == 0 && is_aligned16(a.x) && is_aligned16(a.s0) &&
                   is_aligned16(a.dy) && is_aligned16(a.dst) && is_aligned16(a.y) && is_aligned16(a.st) && is_aligned16(a.weight);
  cudaStream_t st = (cudaStream_t)stream;
  if (a.d.dtype == GDR_BF16) {
    if (!vec) return launch<__nv_bfloat16, 1, 1>(a, dir, dweight, dbias, st);
    // the backward keeps taps, windows and sums of its channels in registers: four channels fit, eight do not
    return launch<__nv_bfloat16, 8, 4>(a, dir, dweight, dbias, st);
  }
  return vec ? launch<float, 4, 4>(a, dir, dweight, dbias, st) : launch<float, 1, 1>(a, dir, dweight, dbias, st);
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
