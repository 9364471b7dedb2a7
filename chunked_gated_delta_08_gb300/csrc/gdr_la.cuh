// gdr_la.cuh -- what the forms of linear attention with a decay for each head
// share: the pass that all of them run, and how sequences are cut into segments.
//
// One pass.  With rows a_t, b_t (Da channels) and c_t (Dc channels) of one head,
// r = e^g and S a Da x Dc state,
//
//   forwards    S_t = r S_{t-1} + b_t c_t^T,            y_t = S_t^T a_t
//   backwards   R_t = r R_{t+1} + b_t c_t^T,  R_{T+1} = S_in / r,  y_t = R_t^T a_t
//
// and the attention and its three gradients are such passes:
//
//   o  = pass(q, k, v)   from h0                dq = pass(do, v, k)  from h0^T
//   dv = pass(k, q, do)  backwards from dht     dk = pass(v, do, q)  backwards from dht^T
//
// A chunk of n rows (i of 0 .. n-1, in the tokens' order both ways) takes
//
//   y_i  = pscale sum_j r^|i-j| (a_i . b_j) c_j + iscale r^e(i) S^T a_i     j <= i, backwards j >= i
//   S'   = r^n S + wscale sum_j r^w(j) b_j c_j^T
//   e(i) = i + 1,  w(j) = n - 1 - j;    backwards  e(i) = n - 1 - i,  w(j) = j + 1
//
// so that no factor exceeds 1 where g <= 0, and the state at a border of chunks
// is the forward's state there, or that state's gradient.
//
// Segments.  Few heads and long sequences leave multiprocessors idle, so a
// sequence is cut into segments of L tokens: one launch forms each segment's own
// state, one carries them along the sequence, one runs the passes from there.  Of a
// packed batch the lengths are on the device, so the blocks themselves see whether
// its longest sequence is worth that; if not, each sequence is one segment and the
// first launch finds nothing to do.
#pragma once

#include "gdr_layer.cuh"

namespace gdr {
namespace la {

constexpr int C = 64;  // tokens in a chunk

// One operand: [tokens, heads, D], rows ld apart; value head hv reads head hv / group.
struct LaRows {
  const void *p;
  int64_t ld;
  int D, group;
};

struct LaPass {
  LaRows a, b, c;
  void *out;          // [tokens, HV, Dc] contiguous; fp32 where out_f32, else of the inputs' type
  const float *s_in;  // states that the sequences start from, null: zero
  const float *carried;  // in kFromStates, where sequences are cut: the states at the segments' borders
  float *s_out;       // state behind the sequence's last chunk, null: not wanted; in kStates: at the borders
  int64_t si, sj;     // element (i, j) of a Da x Dc state lies at i si + j sj
  float pscale, iscale, wscale;
  int backwards, out_f32;
};

// What a launch does with segments: none (a sequence is one), their own states, the passes from carried states.
enum LaMode { kWhole = 0, kStates = 1, kFromStates = 2 };

struct LaArgs {
  LaPass pass[3];
  const float *g;  // [HV]
  const int64_t *cu;
  int *status;
  int64_t N, T, HV, tokens;
  int64_t KV;    // elements of a state
  int64_t L;     // tokens in a segment, a multiple of C (unused in kWhole)
  int64_t least; // sequences are cut where the longest has more tokens than this
  int64_t slots; // segment slots over all sequences, in kStates borders
  int mode;
};

// Segment slot of (sequence n, its segment s) = first token / L + n + s.  Sequences
// take up disjoint ranges of slots, at least one each, whatever their lengths:
// ceil(len / L) <= last / L - first / L + 1.
__host__ __device__ __forceinline__ int64_t slot_count(int64_t tokens, int64_t N, int64_t L) {
  return tokens / L + N;
}
// The states at the borders between a sequence's segments.  The border at token b has
// index b / L: borders of one sequence are L apart, and the first of the next
// sequence is more than L behind the last of this one, so no two share an index,
// and there are tokens / L + 1 of them however many sequences there are.
__host__ __device__ __forceinline__ int64_t border_count(int64_t tokens, int64_t L) { return tokens / L + 1; }
__device__ __forceinline__ int64_t first_slot(const LaArgs &p, int64_t n) {
  return (p.cu ? p.cu[n] : n * p.T) / p.L + n;
}

// seqlens_ok, and whether sequences are cut.  Every thread of the block calls it.
__device__ __forceinline__ bool sequences_ok(const LaArgs &p, bool &cut) {
  __shared__ unsigned longest;
  cut = p.mode != kWhole;
  if (!p.cu) return true;
  if (threadIdx.x == 0) longest = 0;
  if (!seqlens_ok(p.cu, p.N, p.tokens, p.status)) return false;  // (a barrier)
  if (!cut) return true;
  unsigned most = 0;
  for (int64_t n = threadIdx.x; n < p.N; n += blockDim.x) most = max(most, (unsigned)(p.cu[n + 1] - p.cu[n]));
  if (most > p.least) atomicMax(&longest, most);
  __syncthreads();
  cut = longest > p.least;
  return true;
}

struct Segment {
  int64_t n;         // sequence
  int64_t bos, eos;  // tokens of the segment
  int first, last;   // in the pass's order of time
  bool some;         // false: the slot is not in use
};
__device__ __forceinline__ int64_t segments_in(const LaArgs &p, int64_t len) {
  return len > 0 ? (len + p.L - 1) / p.L : 1;
}
// Every thread of the block calls it.  Uncut, the longest of up to 256 sequences come first, so that none of them starts
// last; more take their own order.
__device__ __forceinline__ Segment segment_of(const LaArgs &p, int64_t slot, bool backwards, bool cut) {
  Segment s;
  if (p.mode == kStates) {
    // Border slot + 1: the segment before it covers token (slot + 1) L - 1.  Its state goes to the border behind it,
    // going back that of the segment behind the border.
    const int64_t t = (slot + 1) * p.L - 1;
    s.some = cut && t < p.tokens;
    if (!s.some) return s;
    s.n = seq_of_token(p.cu, p.N, p.T, t);
    const SeqRange r = seq_range(p.cu, s.n, p.T);
    s.bos = t - (t - r.bos) % p.L;
    s.eos = s.bos + p.L;
    s.some = s.eos < r.eos;
    if (backwards) {
      s.bos = s.eos;
      s.eos = r.eos - s.bos < p.L ? r.eos : s.bos + p.L;
    }
    s.first = s.last = 0;
    return s;
  }
  if (!cut) {
    s.some = slot < p.N;
    if (!s.some) return s;
    s.n = seq_of_rank(p.cu, p.N, slot);
    const SeqRange r = seq_range(p.cu, s.n, p.T);
    s.bos = r.bos;
    s.eos = r.eos;
    s.first = s.last = 1;
    return s;
  }
  int64_t lo = 0, hi = p.N;  // first_slot(lo) <= slot < first_slot(hi)
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (first_slot(p, mid) <= slot) lo = mid;
    else hi = mid;
  }
  const SeqRange r = seq_range(p.cu, lo, p.T);
  const int64_t len = r.eos - r.bos, i = slot - first_slot(p, lo), segs = segments_in(p, len);
  s.n = lo;
  s.bos = r.bos + i * p.L;
  s.eos = i == segs - 1 ? r.eos : s.bos + p.L;
  s.some = i < segs;
  s.first = backwards ? i == segs - 1 : i == 0;
  s.last = backwards ? i == 0 : i == segs - 1;
  return s;
}

// The state that a block starts from (null: zero).
__device__ __forceinline__ const float *entering(const LaArgs &p, const LaPass &q, const Segment &s, int64_t hv) {
  if (p.mode == kStates) return nullptr;
  if (!s.first) return q.carried + ((s.bos / p.L + (q.backwards ? 1 : 0)) * p.HV + hv) * p.KV;
  return q.s_in ? q.s_in + (s.n * p.HV + hv) * p.KV : nullptr;
}
// Where the state that a block ends with goes (null: nowhere).
__device__ __forceinline__ float *leaving(const LaArgs &p, const LaPass &q, const Segment &s, int64_t slot,
                                          int64_t hv) {
  if (!q.s_out || !(p.mode == kStates || s.last)) return nullptr;
  return q.s_out + ((p.mode == kStates ? slot + 1 : s.n) * p.HV + hv) * p.KV;
}

// r^n of a whole number n >= 0; r^0 is 1 for every g, -inf (each token forgets all before it) included.
__device__ __forceinline__ float decay_power(float g, int n) { return n == 0 ? 1.f : expf(g * (float)n); }

// A state's decay over n tokens, S -> S a + S b.  Factors near 1 go by what they lack to it (a = r^n - 1, b = 1), so
// that they are not rounded over and over (r^64 of g = -1e-5, rounded to 24 bits, is off by 4e-5 after 512 chunks);
// those below a half as they are (a = r^n, b = 0), because r^n - 1 is rounded to 2^-25, whatever is left of r^n (at
// g = -0.25, 6 % of r^64, and at -0.3 all of it).
struct Decay {
  float a, b;
};
__device__ __forceinline__ Decay decay_of(float g, int64_t n) {
  if (n == 0) return {0.f, 1.f};
  const float x = g * (float)n;
  return x > -0.6931f ? Decay{expm1f(x), 1.f} : Decay{expf(x), 0.f};  // a NaN stays one
}
__device__ __forceinline__ float decayed(float s, Decay d) { return fmaf(s, d.a, s * d.b); }

// The same over a segment, whose r^n may leave fp32's range where S r^n does not: in two halves, so that both factors
// are in range wherever the product is, and no larger than the largest number, so that S = 0 stays 0.
struct LongDecay {
  Decay first, second;
};
__device__ __forceinline__ LongDecay long_decay_of(float g, int64_t n) {
  if (!(fabsf(g * (float)n) > 64.f)) return {decay_of(g, n), {0.f, 1.f}};
  LongDecay d{decay_of(g, n / 2), decay_of(g, n - n / 2)};
  constexpr float kMost = 3.402823466e38f;
  if (d.first.a > kMost) d.first.a = kMost;
  if (d.second.a > kMost) d.second.a = kMost;
  return d;
}
__device__ __forceinline__ float decayed(float s, LongDecay d) { return decayed(decayed(s, d.first), d.second); }

// The tensor-core form (gdr_la_tc.cu): whether it takes these passes, and its launch.
bool tc_takes(const LaArgs &p, int passes, int dtype);
int launch_tc(const LaArgs &p, int passes, cudaStream_t st);

}  // namespace la
}  // namespace gdr
