// gdr_la.cu -- linear attention with a decay for each head: the entry points,
// the form for every type and size, and the single-token form.
#include <algorithm>

#include "gdr_la.cuh"
#include "gdr_sm100.cuh"

namespace gdr {
namespace la {
namespace {

// --------------------------------------------------------------------- any type, any size
// One block per (segment, value head, 32 columns of c), 8 warps.  Operands lie in
// shared memory in fp32; products are warp-level tensor-core products of values
// split into two tf32 parts (2^-21 of a product is lost; bf16 inputs are exact in one
// part).  The tensor cores cut off what they add to an accumulator, so the large
// products and the small ones have one each, and a chunk's part of the state is
// summed by itself: 4e-7 of a state after 16384 tokens, where one accumulator for
// all left 5e-6.  Rows past the segment's end and channels past the width are zeros in
// shared memory.  Two blocks a multiprocessor are bound by issue (40 %) and the
// tensor pipe (37 %): 2 x 2048 x 8 x 64 fp32 take 82 us in three launches.
constexpr int kThreads = 256;
constexpr int kCols = 32;       // columns of c in a block
constexpr int LDC = kCols + 4;  // row strides in shared memory, chosen off multiples of 32 banks
constexpr int LDP = C + 4;

inline int pad16(int n) { return (n + 15) & ~15; }
inline size_t smem_bytes(int Da) {
  const int D = pad16(Da);
  return sizeof(float) * ((size_t)2 * C * (D + 4) + C * LDC + C * LDP + D * LDC + 2 * (C + 4));
}

// rows x D elements of one head into dst [C][ld], zeros past `rows` and from D to Dp.
template <typename T>
__device__ __forceinline__ void load_tile(float *dst, int ld, const LaRows &r, int64_t row0, int head, int rows,
                                          int col0, int cols, int Dp, bool vec) {
  const T *src = static_cast<const T *>(r.p) + row0 * r.ld + (int64_t)(head / r.group) * r.D + col0;
  if (vec) {
    const int per = Dp / 4;
    for (int i = threadIdx.x; i < C * per; i += kThreads) {
      const int row = i / per, c = i % per * 4;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (row < rows && c < cols) load4(src + row * r.ld + c, v);  // cols is a multiple of 4
      store4(dst + row * ld + c, v);
    }
  } else {
    for (int i = threadIdx.x; i < C * Dp; i += kThreads) {
      const int row = i / Dp, c = i % Dp;
      dst[row * ld + c] = row < rows && c < cols ? to_f32(src[row * r.ld + c]) : 0.f;
    }
  }
}

// x in tf32 parts: hi its first 11 bits, lo 11 of the 13 that are left (2^-22 of x is lost; cut off, not rounded:
// adding to the bits would turn some NaN into numbers).  EXACT: x has no more than 8 bits.
template <bool EXACT>
struct Split {
  uint32_t hi, lo;
  __device__ __forceinline__ explicit Split(float x) {
    if constexpr (EXACT) {
      hi = __float_as_uint(x);
      lo = 0;
    } else {
      hi = __float_as_uint(x) & 0xffffe000u;
      lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
    }
  }
};
// large += hi hi, small += the other products; a 16 x 8, b 8 x 8 fragments.
template <bool EA, bool EB>
__device__ __forceinline__ void mma_parts(float (&large)[4], float (&small)[4], const Split<EA> (&a)[4],
                                          const Split<EB> (&b)[2]) {
  if constexpr (!EA && !EB) sm100::mma_tf32(small, a[0].lo, a[1].lo, a[2].lo, a[3].lo, b[0].lo, b[1].lo);
  if constexpr (!EA) sm100::mma_tf32(small, a[0].lo, a[1].lo, a[2].lo, a[3].lo, b[0].hi, b[1].hi);
  if constexpr (!EB) sm100::mma_tf32(small, a[0].hi, a[1].hi, a[2].hi, a[3].hi, b[0].lo, b[1].lo);
  sm100::mma_tf32(large, a[0].hi, a[1].hi, a[2].hi, a[3].hi, b[0].hi, b[1].hi);
}
// NT tiles of 8 columns: acc += a b over K, K a multiple of 8; fa(i, k) of 16 rows, fb(k, j) of 8 NT columns.
template <bool EA, bool EB, int NT, typename FA, typename FB>
__device__ __forceinline__ void tile_product(float (&acc)[NT][4], int K, FA fa, FB fb) {
  const int lane = threadIdx.x & 31, gr = lane >> 2, tg = lane & 3;
  float small[NT][4] = {};
#pragma unroll 2
  for (int k = 0; k < K; k += 8) {
    const Split<EA> a[4] = {Split<EA>(fa(gr, k + tg)), Split<EA>(fa(gr + 8, k + tg)), Split<EA>(fa(gr, k + tg + 4)),
                            Split<EA>(fa(gr + 8, k + tg + 4))};
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const Split<EB> b[2] = {Split<EB>(fb(k + tg, 8 * j + gr)), Split<EB>(fb(k + tg + 4, 8 * j + gr))};
      mma_parts(acc[j], small[j], a, b);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] += small[j][e];
}

template <typename T>
__device__ __forceinline__ bool vec4_ok(const LaRows &r) {
  return r.D % 4 == 0 && r.ld % 4 == 0 && (reinterpret_cast<uintptr_t>(r.p) & (4 * sizeof(T) - 1)) == 0;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) la_any_kernel(const __grid_constant__ LaArgs p) {
  extern __shared__ __align__(16) float sm[];
  bool cut;
  if (!sequences_ok(p, cut)) return;
  const LaPass &q = p.pass[blockIdx.z];
  const int64_t hv = blockIdx.x % p.HV, slot = blockIdx.x / p.HV;
  const int Da = q.a.D, Dc = q.c.D, col0 = blockIdx.y * kCols;
  if (col0 >= Dc) return;
  const bool bw = q.backwards;
  const Segment s = segment_of(p, slot, bw, cut);
  if (!s.some) return;
  const int D = (Da + 15) & ~15, LDA = D + 4, cols = min(kCols, Dc - col0);
  float *A = sm, *B = A + C * LDA, *Cm = B + C * LDA, *P = Cm + C * LDC, *S = P + C * LDP, *pw = S + D * LDC,
        *wt = pw + C + 4;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gr = lane >> 2, tg = lane & 3;
  const float g = p.g[hv];
  const bool va = vec4_ok<T>(q.a), vb = vec4_ok<T>(q.b), vc = vec4_ok<T>(q.c);

  for (int i = tid; i <= C; i += kThreads) pw[i] = decay_power(g, i);
  // the state the segment starts from
  const float *from = entering(p, q, s, hv);
  for (int i = tid; i < D * kCols; i += kThreads) {
    const int r = i / kCols, c = i % kCols;
    S[r * LDC + c] = from && r < Da && c < cols ? from[r * q.si + (col0 + c) * q.sj] : 0.f;
  }
  const int64_t len = s.eos - s.bos;
  const int chunks = (int)((len + C - 1) / C);
  for (int u = 0; u < chunks; ++u) {
    const int64_t t0 = s.bos + (int64_t)(bw ? chunks - 1 - u : u) * C;
    const int n = (int)min((int64_t)C, s.eos - t0);
    __syncthreads();
    if (p.mode != kStates) load_tile<T>(A, LDA, q.a, t0, (int)hv, n, 0, Da, D, va);
    load_tile<T>(B, LDA, q.b, t0, (int)hv, n, 0, Da, D, vb);
    load_tile<T>(Cm, LDC, q.c, t0, (int)hv, n, col0, cols, kCols, vc);
    if (tid < C) wt[tid] = tid < n ? pw[bw ? tid + 1 : n - 1 - tid] * q.wscale : 0.f;
    __syncthreads();
    constexpr bool EX = sizeof(T) == 2;
    if (p.mode != kStates) {
      // P = (A B^T) r^|i-j|: a warp takes 16 rows and 32 columns
      const int r0 = (warp >> 1) * 16, c0 = (warp & 1) * 32;
      float acc[4][4] = {};
      tile_product<EX, EX>(acc, D, [&](int i, int k) { return A[(r0 + i) * LDA + k]; },
                           [&](int k, int j) { return B[(c0 + j) * LDA + k]; });
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + gr + (e >> 1) * 8, c = c0 + 8 * j + 2 * tg + (e & 1);
          const bool in = bw ? c >= r : c <= r;
          P[r * LDP + c] = in ? acc[j][e] * (pw[abs(r - c)] * q.pscale) : 0.f;
        }
      }
      // y = iscale r^e(i) A S + P C: a warp takes 16 rows and 16 columns
      const int oc = (warp & 1) * 16;
      float o[2][4] = {}, o1[2][4] = {};
      tile_product<EX, false>(o, D, [&](int i, int k) { return A[(r0 + i) * LDA + k]; },
                              [&](int k, int j) { return S[k * LDC + oc + j]; });
      __syncthreads();
      tile_product<false, EX>(o1, C, [&](int i, int k) { return P[(r0 + i) * LDP + k]; },
                              [&](int k, int j) { return Cm[k * LDC + oc + j]; });
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + gr + (e >> 1) * 8, c = oc + 8 * j + 2 * tg + (e & 1);
          if (r < n && c < cols) {
            const float y = fmaf(o[j][e], pw[bw ? n - 1 - r : r + 1] * q.iscale, o1[j][e]);
            const int64_t to = ((t0 + r) * p.HV + hv) * Dc + col0 + c;
            if (q.out_f32) static_cast<float *>(q.out)[to] = y;
            else static_cast<T *>(q.out)[to] = from_f32<T>(y);
          }
        }
    }
    // S = r^n S + (w B)^T C: a warp takes rows of S, 16 at a time
    const Decay decay = decay_of(g, n);
    for (int r0 = warp * 16; r0 < D; r0 += 8 * 16) {
      float acc[4][4] = {};
      tile_product<false, EX>(acc, C, [&](int i, int k) { return B[k * LDA + r0 + i] * wt[k]; },
                              [&](int k, int j) { return Cm[k * LDC + j]; });
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float &at = S[(r0 + gr + (e >> 1) * 8) * LDC + 8 * j + 2 * tg + (e & 1)];
          at = decayed(at, decay) + acc[j][e];
        }
    }
  }
  float *to = leaving(p, q, s, slot, hv);
  if (!to) return;
  __syncthreads();
  for (int i = tid; i < Da * kCols; i += kThreads) {
    const int r = i / kCols, c = i % kCols;
    if (c < cols) to[r * q.si + (col0 + c) * q.sj] = S[r * LDC + c];
  }
}

// ------------------------------------------------------------------------------ carry, sums
// The states at the borders, in place of the segments' own: over a sequence's borders
// in the pass's order, S = r^len S + own.  A thread has VEC elements of a head's state, and
// eight borders' of them on their way at once (74 segments one after the other took 50 us).
// Window j of L tokens, j >= 1: of the sequences that start in ((j - 1) L ..< j L) only the last can have
// a border, and its first one has index j.
template <int VEC>
__global__ void __launch_bounds__(256) la_carry_kernel(const __grid_constant__ LaArgs p) {
  bool cut;
  if (!sequences_ok(p, cut) || !cut) return;
  const LaPass &q = p.pass[blockIdx.z];
  const int64_t e = ((int64_t)blockIdx.y * 256 + threadIdx.x) * VEC;
  const int64_t j = blockIdx.x / p.HV + 1, hv = blockIdx.x % p.HV;
  if (e >= p.KV) return;
  const int64_t n = seq_of_token(p.cu, p.N, p.T, j * p.L - 1);
  const SeqRange r = seq_range(p.cu, n, p.T);
  const int64_t segs = segments_in(p, r.eos - r.bos);
  if (r.bos < (j - 1) * p.L || segs < 2) return;
  const float g = p.g[hv];
  float S[VEC] = {};
  if (q.s_in) load_vec<VEC>(q.s_in + (n * p.HV + hv) * p.KV + e, S);
  const int64_t step = p.HV * p.KV * (q.backwards ? -1 : 1);
  float *own = q.s_out + ((j + (q.backwards ? segs - 2 : 0)) * p.HV + hv) * p.KV + e;
  const LongDecay full = long_decay_of(g, p.L), tail = long_decay_of(g, r.eos - r.bos - (segs - 1) * p.L);
  constexpr int kAhead = 8;
  for (int64_t u0 = 0; u0 < segs - 1; u0 += kAhead, own += kAhead * step) {
    float mine[kAhead][VEC];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (u0 + i < segs - 1) load_vec<VEC>(own + i * step, mine[i]);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (u0 + i < segs - 1) {
        // the ragged segment is a sequence's last: going back, the first of the pass
        const LongDecay decay = q.backwards && u0 + i == 0 ? tail : full;
#pragma unroll
        for (int k = 0; k < VEC; ++k) S[k] = decayed(S[k], decay) + mine[i][k];
        store_vec<VEC>(own + i * step, S);
      }
    }
  }
}

// out [M, H, D] = sums over groups of G value heads of part [M, H G, D], in order; VEC elements to a thread.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) la_sum_kernel(const float *part0, const float *part1, T *out0, T *out1,
                                                     int64_t n, int G, int D, SeqCheck check) {
  if (!seqlens_ok(check)) return;
  const float *part = blockIdx.y ? part1 : part0;
  T *out = blockIdx.y ? out1 : out0;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * VEC;
  if (i >= n) return;
  const float *src = part + i / D * G * D + i % D;
  float s[VEC];
  load_vec<VEC>(src, s);
#pragma unroll 4
  for (int j = 1; j < G; ++j) {
    float v[VEC];
    load_vec<VEC>(src + (int64_t)j * D, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] += v[e];
  }
  store_vec<VEC>(out + i, s);
}
template <typename T>
int launch_sum(const float *part0, const float *part1, void *out0, void *out1, int64_t n, int G, int D,
               const SeqCheck &check, cudaStream_t st) {
  const bool vec = D % 4 == 0 && is_aligned16(out0) && is_aligned16(out1);
  const auto kernel = vec ? la_sum_kernel<T, 4> : la_sum_kernel<T, 1>;
  const dim3 grid((unsigned)cdiv(n, vec ? 1024 : 256), 2);
  kernel<<<grid, 256, 0, st>>>(part0, part1, (T *)out0, (T *)out1, n, G, D, check);
  return launched("la_sum_kernel");
}

// -------------------------------------------------------------------------------- host side
// How sequences are cut: p.L (0: not) and p.least.  A block walks a sequence chunk by chunk, `wave`
// blocks at a time (a tensor-core block takes 1.7 us a chunk, one of the other form some 9 at 64 fp32 channels).  Rows of
// more than 128 channels leave room for one block of the other form on a multiprocessor, not two; these constants
// were measured with two, and with one in their place as many calls became slower as faster (bf16: 4 x 4096 x 4 heads x
// 256 x 256 1734 -> 1408 us, but 32768 x 4 3730 -> 4103, its backward 8103 -> 9833, and that of 16384 x 2 heads x 128 x
// 256 1333 -> 1861).  Uncut, a launch takes as long as its longest sequence, or its waves of whole sequences.  Cut, the work
// spreads evenly, but forming the segments' states and ragged waves make it 2.2 times as much (16384 x 32
// heads in 7 sequences, 94 chunks the longest: 168 us uncut, 223 cut, when measured for this; 8192 x 16 heads 69 us cut), and
// two more launches take the time of `launches` chunks; a segment has at least `shortest` of them.
void cut(LaArgs &p, int blocks_per_pair, int wave, int launches, int shortest) {
  const int64_t blocks = p.HV * blocks_per_pair;                // to a sequence
  const int64_t even = cdiv(cdiv(p.tokens, C) * blocks, wave);  // chunks of work to a block of a wave
  p.least = C * (launches + 11 * std::max<int64_t>(even, 4) / 5);
  p.L = 0;
  const int64_t longest = p.cu ? p.tokens : cdiv(p.N * blocks, wave) * p.T;
  if (p.N == 0 || longest <= p.least) return;
  // Where all sequences are alike, all segments in one wave; else half a wave's share, which packs better.
  const int64_t alike = p.cu ? (p.N == 1 ? p.tokens : 0) : p.T, each = wave / (p.N * blocks);
  const int64_t chunks = alike && each ? cdiv(cdiv(alike, C), each) : cdiv(even, 2);
  p.L = C * std::max<int64_t>(shortest, chunks);
  if (p.L >= (alike ? alike : p.tokens)) p.L = 0;
}

template <typename T>
int launch_any(const LaArgs &p, int passes, cudaStream_t st) {
  int Da = 0, Dc = 0;
  for (int i = 0; i < passes; ++i) {
    Da = std::max(Da, p.pass[i].a.D);
    Dc = std::max(Dc, p.pass[i].c.D);
  }
  const size_t smem = smem_bytes(Da);
  const cudaError_t e = cudaFuncSetAttribute(la_any_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute(la_any_kernel)");
  const int64_t items = std::max<int64_t>(1, (p.mode == kWhole ? p.N : p.slots) * p.HV);
  if (items > 0x7fffffff) return set_error(GDR_ERR_SHAPE, "too many sequences and heads for one launch");
  la_any_kernel<T><<<dim3((unsigned)items, (unsigned)cdiv(Dc, kCols), passes), kThreads, smem, st>>>(p);
  return launched("la_any_kernel");
}

int launch(const LaArgs &p, int passes, int dtype, bool tc, cudaStream_t st) {
  if (tc) return launch_tc(p, passes, st);
  return dtype == GDR_BF16 ? launch_any<__nv_bfloat16>(p, passes, st) : launch_any<float>(p, passes, st);
}

// Runs `passes` of p; states (nstates of them, in passes st_pass, with natural strides) are
// formed and carried first where sequences are cut.  from[i]: which state pass i starts from.
int run(LaArgs p, int passes, const LaPass *st_pass, int nstates, const int *from, int dtype, cudaStream_t st) {
  const bool tc = tc_takes(p, passes, dtype);
  p.mode = kWhole;
  int widest = 1;
  for (int i = 0; i < passes; ++i) widest = std::max(widest, (int)cdiv(p.pass[i].c.D, kCols));
  if (tc) cut(p, passes, kSMs, 10, 4);
  else cut(p, passes * widest, 2 * kSMs, 3, 2);
  if (!p.L) return launch(p, passes, dtype, tc, st);
  p.slots = slot_count(p.tokens, p.N, p.L);
  const int64_t borders = border_count(p.tokens, p.L) - 1, one = (borders + 1) * p.HV * p.KV;
  if (borders * p.HV > 0x7fffffff) return set_error(GDR_ERR_SHAPE, "too many tokens and heads for one launch");
  char *base = nullptr;
  int rc = scratch_begin(sizeof(float) * (size_t)(one * nstates), st, "linear attention states", &base);
  if (rc != GDR_OK) return rc;
  LaArgs s = p;
  s.mode = kStates;
  s.slots = borders;
  for (int i = 0; i < nstates; ++i) {
    s.pass[i] = st_pass[i];
    s.pass[i].s_out = (float *)base + i * one;
  }
  rc = launch(s, nstates, dtype, tc_takes(s, nstates, dtype), st);
  if (rc == GDR_OK) {
    bool vec = p.KV % 4 == 0;
    for (int i = 0; i < nstates; ++i) vec = vec && is_aligned16(s.pass[i].s_in);
    const auto kernel = vec ? la_carry_kernel<4> : la_carry_kernel<1>;
    kernel<<<dim3((unsigned)(borders * p.HV), (unsigned)cdiv(p.KV, vec ? 1024 : 256), nstates), 256, 0, st>>>(s);
    rc = launched("la_carry_kernel");
  }
  p.mode = kFromStates;
  for (int i = 0; i < passes; ++i) p.pass[i].carried = (float *)base + from[i] * one;
  if (rc == GDR_OK) rc = launch(p, passes, dtype, tc, st);
  return scratch_end(base, st, "linear attention states", rc);
}

int validate(const gdr_la_desc *d, const int64_t *cu, bool step) {
  if (!d) return set_error(GDR_ERR_NULLPTR, "desc is NULL");
  if (d->dtype != GDR_F32 && d->dtype != GDR_BF16) return set_error(GDR_ERR_DTYPE, "dtype must be GDR_F32 or GDR_BF16");
  if (d->flags) return set_error(GDR_ERR_DTYPE, "unknown bits in flags");
  constexpr int64_t kMost = 0x7fffffff;
  if (d->B < 0 || d->T < 0 || d->N < 0 || d->N > kMost || d->B > kMost || d->T > kMost ||
      (d->T > 0 && d->B > kMost / d->T))
    return set_error(GDR_ERR_SHAPE, "B, T and N must be >= 0, N and B * T below 2^31");
  if (d->H < 1 || d->HV < 1 || d->HV % d->H != 0 || d->HV > 65535)
    return set_error(GDR_ERR_SHAPE, "HV must be a multiple of H, at most 65535");
  if (d->K < 1 || d->K > 256 || d->V < 1 || d->V > 256) return set_error(GDR_ERR_SHAPE, "K and V must be in [1, 256]");
  if (d->ld_q < d->H * d->K || d->ld_k < d->H * d->K || d->ld_v < d->HV * d->V || d->ld_do < d->HV * d->V)
    return set_error(GDR_ERR_SHAPE, "leading dimensions must be at least H * K, or HV * V");
  if (d->ld_q > kMost || d->ld_k > kMost || d->ld_v > kMost || d->ld_do > kMost)
    return set_error(GDR_ERR_SHAPE, "leading dimensions must be below 2^31");
  if (!(d->scale - d->scale == 0.f)) return set_error(GDR_ERR_SHAPE, "scale must be finite");
  if (step) return d->T == 1 ? GDR_OK : set_error(GDR_ERR_SHAPE, "a step takes one token per row: T must be 1");
  if (cu) {
    if (d->B != 1) return set_error(GDR_ERR_SHAPE, "cu_seqlens requires B == 1");
  } else if (d->N != d->B) {
    return set_error(GDR_ERR_SHAPE, "N must equal B when cu_seqlens is NULL");
  }
  return GDR_OK;
}

LaArgs base_args(const gdr_la_desc &d, const float *g, const int64_t *cu, int *status) {
  LaArgs p{};
  p.g = g;
  p.cu = cu;
  p.status = status;
  p.N = d.N;
  p.T = d.T;
  p.HV = d.HV;
  p.tokens = d.B * d.T;
  p.KV = d.K * d.V;
  return p;
}

// ------------------------------------------------------------------------------ single tokens
// One block per (row, value head, run of columns) walks its part of the K x V state once:
// S = r S + k v^T is written back and o = scale S^T q summed on the way.  Eight bytes of
// state a multiply-add: HBM bound.  A thread keeps VEC columns; the partial sums of o of
// a block's row groups meet in shared memory, in order.  256 x 32 heads of 128 x 128 take 168 us, 97 % of the
// copy rate (with one row on its way after the other 197).
template <typename T, int VEC>
__global__ void __launch_bounds__(256) la_step_kernel(gdr_la_desc d, const T *q, const T *k, const T *v, const float *g,
                                                      const int32_t *slots, float *state, T *o, int *status, int run) {
  __shared__ float sq[256], sk[256];
  __shared__ __align__(16) float part[256 * VEC];
  const int K = (int)d.K, V = (int)d.V, tid = threadIdx.x;
  const int64_t row = blockIdx.x / d.HV, hv = blockIdx.x % d.HV, h = hv / (d.HV / d.H);
  const int first = blockIdx.y * run, cols = min(run, V - first);
  int64_t slot = slots ? slots[row] : row;
  if (slot >= d.N) {
    if (tid == 0 && hv == 0 && first == 0) raise_status(status, GDR_ERR_SLOTS);
    slot = -1;
  }
  T *to = o + (row * d.HV + hv) * V + first;
  if (slot < 0) {
    for (int c = tid; c < cols; c += 256) to[c] = from_f32<T>(0.f);
    return;
  }
  if (tid < K) {
    sq[tid] = to_f32(q[row * d.ld_q + h * K + tid]) * d.scale;
    sk[tid] = to_f32(k[row * d.ld_k + h * K + tid]);
  }
  __syncthreads();
  const int across = (cols + VEC - 1) / VEC, groups = 256 / across;  // cols <= 256
  const int c = tid % across * VEC, r0 = tid / across;
  const Decay decay = decay_of(g[hv], 1);
  float acc[VEC] = {};
  if (r0 < groups) {
    float vv[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) vv[i] = to_f32(v[row * d.ld_v + hv * V + first + c + i]);
    float *S = state + (slot * d.HV + hv) * (int64_t)K * V + first + c;
    constexpr int U = 4;  // rows on their way at once
    for (int i0 = r0; i0 < K; i0 += U * groups) {
      float s[U][VEC];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * groups < K) load_vec<VEC>(S + (int64_t)(i0 + u * groups) * V, s[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * groups;
        if (i < K) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            s[u][j] = fmaf(sk[i], vv[j], decayed(s[u][j], decay));
            acc[j] = fmaf(sq[i], s[u][j], acc[j]);
          }
          store_vec<VEC>(S + (int64_t)i * V, s[u]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) part[tid * VEC + j] = acc[j];
  __syncthreads();
  for (int i = tid; i < cols; i += 256) {
    float s = 0.f;
    for (int gq = 0; gq < groups; ++gq) s += part[gq * across * VEC + i];
    to[i] = from_f32<T>(s);
  }
}

template <typename T>
int launch_step(const gdr_la_desc &d, const void *q, const void *k, const void *v, const float *g, const int32_t *slots,
                float *state, void *o, int *status, cudaStream_t st) {
  const int64_t blocks = d.B * d.HV;
  if (blocks > 0x7fffffff) return set_error(GDR_ERR_SHAPE, "too many rows and heads for one launch");
  const bool vec = d.V % 4 == 0 && is_aligned16(state);
  // Few heads in all: runs of 32 columns, whole lines of the state, share a head out over four blocks
  // (1 x 32 x 128 x 128 in a graph: 5.5 us in whole heads, 2.8 so).
  const int run = blocks < 2 * kSMs ? 32 : 256;
  const auto kernel = vec ? la_step_kernel<T, 4> : la_step_kernel<T, 1>;
  const dim3 grid((unsigned)blocks, (unsigned)cdiv(d.V, run));
  kernel<<<grid, 256, 0, st>>>(d, (const T *)q, (const T *)k, (const T *)v, g, slots, state, (T *)o, status, run);
  return launched("la_step_kernel");
}

}  // namespace
}  // namespace la
}  // namespace gdr

using namespace gdr;
using namespace gdr::la;

extern "C" {

int gdr_la_fwd(const gdr_la_desc *desc, const void *q, const void *k, const void *v, const float *g, const float *h0,
               const int64_t *cu_seqlens, void *o, float *ht, void *stream) {
  int rc = validate(desc, cu_seqlens, false);
  if (rc != GDR_OK) return rc;
  const gdr_la_desc &d = *desc;
  if (d.N == 0 && !cu_seqlens) return GDR_OK;
  if (!g || (d.B * d.T > 0 && (!q || !k || !v || !o)))
    return set_error(GDR_ERR_NULLPTR, "q, k, v, g and o must be non-NULL");
  int *status = current_status_word(&rc);
  if (!status) return rc;
  LaArgs p = base_args(d, g, cu_seqlens, status);
  const int G = (int)(d.HV / d.H);
  const LaRows rq{q, d.ld_q, (int)d.K, G}, rk{k, d.ld_k, (int)d.K, G}, rv{v, d.ld_v, (int)d.V, 1};
  p.pass[0] = {rq, rk, rv, o, h0, nullptr, ht, d.V, 1, d.scale, d.scale, 1.f, 0, 0};
  const LaPass state = p.pass[0];
  const int from[1] = {0};
  return run(p, 1, &state, 1, from, d.dtype, (cudaStream_t)stream);
}

int gdr_la_bwd(const gdr_la_desc *desc, const void *q, const void *k, const void *v, const float *g, const float *h0,
               const int64_t *cu_seqlens, const void *d_o, const float *dht, void *dq, void *dk, void *dv, float *dh0,
               void *stream) {
  int rc = validate(desc, cu_seqlens, false);
  if (rc != GDR_OK) return rc;
  const gdr_la_desc &d = *desc;
  if (d.N == 0 && !cu_seqlens) return GDR_OK;
  if (!g || (d.B * d.T > 0 && (!q || !k || !v || !d_o || !dq || !dk || !dv)))
    return set_error(GDR_ERR_NULLPTR, "q, k, v, g, d_o, dq, dk and dv must be non-NULL");
  int *status = current_status_word(&rc);
  if (!status) return rc;
  LaArgs p = base_args(d, g, cu_seqlens, status);
  const cudaStream_t st = (cudaStream_t)stream;
  const int G = (int)(d.HV / d.H);
  const int64_t n = d.B * d.T * d.HV * d.K;
  // grouped value heads: their parts of dq and dk meet in fp32
  char *base = nullptr;
  if (G > 1 && n > 0) {
    rc = scratch_begin(sizeof(float) * 2 * (size_t)n, st, "parts of dq and dk", &base);
    if (rc != GDR_OK) return rc;
  }
  float *pq = (float *)base, *pk = base ? pq + n : nullptr;
  const LaRows rq{q, d.ld_q, (int)d.K, G}, rk{k, d.ld_k, (int)d.K, G}, rv{v, d.ld_v, (int)d.V, 1},
      rd{d_o, d.ld_do, (int)d.V, 1};
  const int parts = base != nullptr;
  // passes of the same direction side by side: dk and dv read the same rows
  p.pass[0] = {rk, rq, rd, dv, dht, nullptr, dh0, d.V, 1, d.scale, 1.f, d.scale, 1, 0};
  p.pass[1] = {rv, rd, rq, parts ? pk : dk, dht, nullptr, nullptr, 1, d.V, d.scale, 1.f, d.scale, 1, parts};
  p.pass[2] = {rd, rv, rk, parts ? pq : dq, h0, nullptr, nullptr, 1, d.V, d.scale, d.scale, 1.f, 0, parts};
  LaPass states[2] = {p.pass[0], {rq, rk, rv, nullptr, h0, nullptr, nullptr, d.V, 1, d.scale, d.scale, 1.f, 0, 0}};
  const int from[3] = {0, 0, 1};
  rc = run(p, 3, states, 2, from, d.dtype, st);
  if (!base) return rc;
  if (rc == GDR_OK) {
    const SeqCheck check{cu_seqlens, d.N, d.B * d.T, status};
    rc = d.dtype == GDR_BF16 ? launch_sum<__nv_bfloat16>(pq, pk, dq, dk, n / G, G, (int)d.K, check, st)
                             : launch_sum<float>(pq, pk, dq, dk, n / G, G, (int)d.K, check, st);
  }
  return scratch_end(base, st, "parts of dq and dk", rc);
}

int gdr_la_step(const gdr_la_desc *desc, const void *q, const void *k, const void *v, const float *g,
                const int32_t *slots, float *state, void *o, void *stream) {
  int rc = validate(desc, nullptr, true);
  if (rc != GDR_OK) return rc;
  if (desc->B == 0) return GDR_OK;
  if (!q || !k || !v || !g || !state || !o)
    return set_error(GDR_ERR_NULLPTR, "q, k, v, g, state and o must be non-NULL");
  int *status = current_status_word(&rc);
  if (!status) return rc;
  const cudaStream_t st = (cudaStream_t)stream;
  return desc->dtype == GDR_BF16 ? launch_step<__nv_bfloat16>(*desc, q, k, v, g, slots, state, o, status, st)
                                 : launch_step<float>(*desc, q, k, v, g, slots, state, o, status, st);
}

}  // extern "C"
