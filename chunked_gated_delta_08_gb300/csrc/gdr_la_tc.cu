// gdr_la_tc.cu -- linear attention with a decay for each head on the sm_103a
// tensor cores: the passes of gdr_la.cuh for bf16 rows of up to 128 channels.
//
// One block per (segment, value head, pass) walks its tokens in chunks of 64 with the
// state on chip: rows of a, b and c are read once, y is written once.  Per chunk of n
// rows, with r = e^g and the state held transposed, Dc x Da, in tensor memory:
//
//   Sc   = A B^T                                    M=64  N=64   K=Da
//   P_ij = pscale r^|i-j| Sc_ij  (j <= i; backwards j >= i), bf16
//   B'_j = wscale r^w(j) B_j = hi + lo, two bf16    (2^-17 of each product: states leave in fp32, and hi alone would
//                                                    leave 2^-9 in them; it saves 3 % where none leaves)
//   O1^T = C^T P^T                                  M=128 N=64   K=64
//   O2^T = S^T A^T, S^T as bf16 in tensor memory    M=128 N=64   K=Da
//   U^T  = C^T B'hi + C^T B'lo                      M=128 N=Da K=64
//   S^T  = r^n S^T + U^T                            by the state's warps, in fp32
//   y_i  = O1_i + iscale r^e(i) O2_i
//
// Every factor is a power of r with an exponent that the place in the chunk gives, so
// the threads keep them in registers; only a ragged last chunk works them out anew.
//
// The tensor cores cut off what they add to an accumulator: a state that all chunks are added to there loses
// 1.6e-4 of itself over 32768 tokens of one sign and 7e-4 over 131072.  So U has a buffer of its own,
// and the state loses 3e-7 and 6e-7 (4 x 4096 x 32 x 128: forward 110 -> 115 us, backward 318 -> 326).  That takes the columns of
// the second scores and the second copy of the state; outputs' MMAs in the order O2, O1 took 4 % longer.
//
// What follows one chunk after the other is U's MMAs, then their reading by the state's warps (0-7), which make
// the next bf16 copy meanwhile.  An issuing thread stands still for some 200 cycles at each burst of MMAs and each
// commit, so the three kinds have a thread each (one for all took 1.8 us a chunk where three took 1.6).
//
// Warp roles (896 threads):
//   warps 0-7    state: S = r^n S + U in tensor memory, its bf16 copy
//   warps 8-15   scores: P, B' (over B in place, its lower half beside), rows past a ragged end cleared
//   warps 16-23  output: y through shared memory and a tensor store
//   warp 24      producer: TMA loads into a ring of three stages, six where rows have up to 64 channels
//   warp 25      issues the scores' MMAs
//   warp 26      issues U's
//   warp 27      issues the outputs'
// Hand-offs are mbarriers.  Every wait is bounded (about two seconds): where one runs out
// the block's error flag makes all others return at once, the producer and the MMA threads
// stop, the rest run to their end on what is there (in bounds), the block lets its copies
// and MMAs finish, frees its tensor memory and reports GDR_ERR_TIMEOUT.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "gdr_fused_common.cuh"
#include "gdr_la.cuh"
#include "gdr_sm100.cuh"

namespace gdr {
namespace la {
namespace {

using namespace sm100;
using fused::ld_sw128_chunk;
using fused::st_sw128_chunk;
using fused::sw128_chunk_off;

constexpr int kTcThreads = 896;
constexpr int kProducer = 24, kScoreMma = 25, kStateMma = 26;  // and one more for the outputs' MMAs
constexpr int kBarOut = 1;  // named barrier of the output warps

// Shared memory, from a 1024-byte aligned base.  A tile is one panel of 64 rows x 64 channels where no row has more
// than 64, else two; a stage waits in the ring from its load to its output, three periods and more, so the smaller
// ones get six instead of three (4 x 4096 x 32 x 64: forward 82 -> 76 us, backward 228 -> 206 us).
constexpr uint32_t SZ_PANEL = 8192;
template <int PANELS>
struct Layout {
  static constexpr int kStages = 6 / PANELS;
  static constexpr uint32_t SZ_TILE = PANELS * SZ_PANEL;
  static constexpr uint32_t SZ_STAGE = 3 * SZ_TILE;            // A | B | C
  static constexpr uint32_t OFF_LO = kStages * SZ_STAGE;       // lower parts of B', two buffers
  static constexpr uint32_t OFF_P = OFF_LO + 2 * SZ_TILE;      // P, two buffers
  static constexpr uint32_t OFF_Y = OFF_P + 2 * SZ_PANEL;      // y on its way out: two buffers of bf16, one of fp32
  static constexpr uint32_t OFF_SMALL = OFF_Y + 2 * SZ_TILE;
};
constexpr int kMostStages = 6;

// TMEM columns
constexpr uint32_t TM_SC = 0, TM_O = 64 /* O1, O2 */, TM_S = 192, TM_U = 320, TM_SB = 448, TM_COLS = 512;

struct Small {
  float pw[C + 4];  // r^0 .. r^64
  uint64_t full[kMostStages], empty[kMostStages];
  // (a stage is empty when its chunk's state and output MMAs are done, which frees P and B' too)
  uint64_t b_sc, b_u, b_o, b_final[3];  // MMAs done
  // arrivals of eight warps: P, B', the state's copy; Sc, U, O1 and O2 read
  uint64_t b_p[2], b_bs[2], b_sb, b_scfree, b_ufree, b_ofree;
  uint32_t tmem_slot;
  int err;
};
template <int PANELS>
constexpr uint32_t smem_bytes() {
  return Layout<PANELS>::OFF_SMALL + sizeof(Small) + 1024;
}
static_assert(smem_bytes<1>() <= 232448 && smem_bytes<2>() <= 232448, "shared memory budget");

__device__ __forceinline__ uint32_t pack_f2(f2 v) {
  float lo, hi;
  f2_split(v, lo, hi);
  return gdr::pack_bf16(lo, hi);
}

// One thread of a converged warp, in a form that the compiler knows to be one thread.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

constexpr uint64_t kTimeout = 1ull << 32;  // cycles: about two seconds at the GB300's clocks

// Waits for the phase of the given parity; returns without it once the block's error flag is set, which a wait
// that runs out of time does.
__device__ __forceinline__ void wait_or_err(uint32_t bar, uint32_t parity, volatile int *err) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = clock64();
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
    if ((i & 15u) == 0) {
      if (*err) return;
      if ((uint64_t)clock64() - t0 > kTimeout) {
        *err = 1;
        return;
      }
    }
  }
}

// Waits until at most N of the thread's bulk stores still read shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

struct Maps {
  CUtensorMap a[3], b[3], c[3], y[3];
};

// PARTS: some of the passes write fp32 parts (grouped value heads); their code costs the others 8 %.
template <bool PARTS, int PANELS>
__global__ void __launch_bounds__(kTcThreads, 1)
    la_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ LaArgs p, int passes) {
  using L = Layout<PANELS>;
  constexpr int kStages = L::kStages;
  constexpr uint32_t SZ_TILE = L::SZ_TILE, SZ_STAGE = L::SZ_STAGE;
  constexpr uint32_t OFF_LO = L::OFF_LO, OFF_P = L::OFF_P, OFF_Y = L::OFF_Y;
  extern __shared__ uint8_t smem_raw[];
  bool cut;
  if (!sequences_ok(p, cut)) return;
  uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Small &S = *reinterpret_cast<Small *>(sm + L::OFF_SMALL);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the passes over one item run side by side: the rows that two of them read come from L2 the second time
  const int pi = (int)(blockIdx.x % passes);
  const int64_t item = blockIdx.x / passes;
  const LaPass &q = p.pass[pi];
  const int64_t hv = item % p.HV, slot = item / p.HV;
  const bool bw = q.backwards, states = p.mode == kStates;
  const Segment s = segment_of(p, slot, bw, cut);
  if (!s.some) return;
  const int Da = q.a.D, Dc = q.c.D, ka = PANELS == 2 && Da > 64 ? 2 : 1, kc = PANELS == 2 && Dc > 64 ? 2 : 1;
  const int64_t len = s.eos - s.bos;
  const int nch = (int)((len + C - 1) / C);
  const float g = p.g[hv];
  auto chunk_start = [&](int c) { return s.bos + (int64_t)(bw ? nch - 1 - c : c) * C; };
  // the segment's last chunk, which may be ragged, and its rows
  const int ragged = bw ? 0 : nch - 1, rest = (int)(len - (int64_t)(nch - 1) * C);
  auto chunk_rows = [&](int c) { return c == ragged ? rest : C; };

  if (tid < C + 1) S.pw[tid] = decay_power(g, tid);
  if (tid == 0) {
    S.err = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&S.full[i]), 1);
      mbar_init(smem_u32(&S.empty[i]), p.mode == kStates ? 1 : 2);
    }
    for (uint64_t *b = &S.b_sc; b <= &S.b_final[2]; ++b) mbar_init(smem_u32(b), 1);
    for (uint64_t *b = S.b_p; b <= &S.b_ofree; ++b) mbar_init(smem_u32(b), 8);
    fence_mbar_init();
  }
  if (tid == 32 * kProducer) {
    if (!states) tma_prefetch_desc(&maps.a[pi]);
    tma_prefetch_desc(&maps.b[pi]);
    tma_prefetch_desc(&maps.c[pi]);
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&S.tmem_slot), TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = S.tmem_slot;
  volatile int *err = &S.err;
  uint8_t *const sLo = sm + OFF_LO, *const sP = sm + OFF_P, *const sY = sm + OFF_Y;
  const uint32_t lane_addr = tbase + ((uint32_t)((warp & 3) * 32) << 16);
  auto wait = [&](uint64_t &bar, uint32_t parity) { wait_or_err(smem_u32(&bar), parity, err); };
  // the same without sleeping, for single threads (eight warps of the state group polling took 7 % longer)
  auto spin = [&](uint64_t &bar, uint32_t parity) { mbar_wait_spin(smem_u32(&bar), parity, err, kTimeout); };
  auto arrive = [&](uint64_t &bar) {  // of a warp
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bar));
  };

  if (warp < 8) {
    // ================================================================ state
    const int j = 32 * (warp & 3) + lane;                 // TMEM lane: channel of c
    const int cols = 32 * ka, col0 = (warp >> 2) * cols;  // this thread's channels of a
    const uint32_t aS = lane_addr + TM_S + col0, aU = lane_addr + TM_U + col0, aSb = lane_addr + TM_SB + col0 / 2;
    const bool mine = j < Dc;
    auto copy = [&](int i0, const float (&r)[16]) {
      uint32_t u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = gdr::pack_bf16(r[2 * i], r[2 * i + 1]);
      tmem_st8(aSb + i0 / 2, u);
    };
    {
      const float *from = mine ? entering(p, q, s, hv) : nullptr;
      if (from) from += j * q.sj;
#pragma unroll 1
      for (int i0 = 0; i0 < cols; i0 += 16) {
        float r[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = from && col0 + i0 + i < Da ? from[(int64_t)(col0 + i0 + i) * q.si] : 0.f;
        tmem_st16(aS + i0, r);
        copy(i0, r);
      }
    }
    tmem_st_wait();
    tc_fence_before();
    arrive(S.b_sb);
    const Decay whole = decay_of(g, C);
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
      const int n = chunk_rows(c);
      const Decay decay = n == C ? whole : decay_of(g, n);
      const bool more = !states && c + 1 < nch;  // chunks that read a copy
      wait(S.b_u, c & 1);
      tc_fence_after();
#pragma unroll
      for (int i0 = 0; i0 < 64; i0 += 16) {
        if (i0 < cols) {
          float r[16], u[16];
          tmem_ld16(aU + i0, u);
          tmem_ld16(aS + i0, r);
          tmem_ld_wait();
          if (i0 == 0 && more) {  // O2 has read the copy
            wait(S.b_o, c & 1);
            tc_fence_after();
          }
          if (i0 + 16 == cols) {
            tc_fence_before();
            arrive(S.b_ufree);
          }
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const f2 x = f2_pack(r[i], r[i + 1]);
            const f2 y = f2_fma(x, f2_both(decay.a), f2_pack(u[i], u[i + 1]));
            f2_split(f2_fma(x, f2_both(decay.b), y), r[i], r[i + 1]);
          }
          if (more) copy(i0, r);
          tmem_st16(aS + i0, r);
        }
      }
      tmem_st_wait();
      if (more) {
        tc_fence_before();
        arrive(S.b_sb);
      }
    }
    float *to = leaving(p, q, s, slot, hv);
    if (to) {
      to += j * q.sj;
#pragma unroll 1
      for (int i0 = 0; i0 < cols; i0 += 16) {
        float r[16];
        tmem_ld16(aS + i0, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (mine && col0 + i0 + i < Da) to[(int64_t)(col0 + i0 + i) * q.si] = r[i];
      }
    }
  } else if (warp < 16) {
    // ================================================================ scores
    const int gt = tid - 256, w = warp & 3, half = (warp - 8) >> 2;
    // this thread's scores: rows r0 and r0 + 8, columns 32 half + 8 b + c0 and the next, b of 0 .. 3
    const int r0 = 16 * w + (lane >> 2), c0 = 2 * (lane & 3);
    float f[4][4];
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r0 + 8 * (e >> 1), c = 32 * half + 8 * b + c0 + (e & 1);
        f[b][e] = (bw ? c >= r : c <= r) ? S.pw[abs(r - c)] * q.pscale : 0.f;
      }
    // of B: a row and a quarter of its channels
    const int row = 16 * w + (lane & 15), part = 2 * half + (lane >> 4);
    const int panel = ka == 2 ? part >> 1 : 0, ch0 = ka == 2 ? 4 * (part & 1) : 2 * part, chunks = 2 * ka;
    const float whole_wt = S.pw[bw ? row + 1 : C - 1 - row] * q.wscale, wscale = q.wscale;
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
      const int st = c % kStages, buf = c & 1;
      const int n = chunk_rows(c);
      uint8_t *tile = sm + st * SZ_STAGE;
      wait(S.full[st], (c / kStages) & 1);
      if (n < C) {  // rows past the end may hold the next sequence
        for (int i = gt; i < (C - n) * 8 * kc; i += 256)
          st_sw128_chunk(tile + 2 * SZ_TILE + (kc == 2 && (i & 8) ? SZ_PANEL : 0), n + (kc == 2 ? i >> 4 : i >> 3),
                         i & 7, make_uint4(0, 0, 0, 0));
      }
      if (c > 1) wait(S.empty[(c - 2) % kStages], ((c - 2) / kStages) & 1);  // the buffers' chunk before is done
      if (!states) {
        wait(S.b_sc, c & 1);
        tc_fence_after();
        float r[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i) tmem_ld_16x256b_x2(lane_addr + TM_SC + 32 * half + 16 * i, r[i]);
        tmem_ld_wait();
        tc_fence_before();
        arrive(S.b_scfree);
        if (n < C) {  // columns past the end: what lies there is not multiplied
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (32 * half + 8 * (k >> 2) + c0 + (k & 1) >= n) r[k >> 3][k & 7] = 0.f;
        }
        uint8_t *P = sP + buf * SZ_PANEL;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float *x = r[b >> 1] + 4 * (b & 1);
          uint8_t *to = P + sw128_chunk_off(r0, 4 * half + b) + 2 * c0;
          *reinterpret_cast<uint32_t *>(to) = pack_f2(f2_mul(f2_pack(x[0], x[1]), f2_pack(f[b][0], f[b][1])));
          *reinterpret_cast<uint32_t *>(to + 1024) = pack_f2(f2_mul(f2_pack(x[2], x[3]), f2_pack(f[b][2], f[b][3])));
        }
        fence_proxy_async_smem();
        arrive(S.b_p[buf]);
      }
      // B' over B (the scores' product has read it), its lower half beside
      const float wt = n == C ? whole_wt : row < n ? S.pw[bw ? row + 1 : n - 1 - row] * wscale : 0.f;
      uint8_t *hi = tile + SZ_TILE + panel * SZ_PANEL, *lo = sLo + buf * SZ_TILE + panel * SZ_PANEL;
      uint4 in[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < chunks) in[i] = row < n ? ld_sw128_chunk(hi, row, ch0 + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < chunks) {
          float v[8];
          unpack8(in[i], v);
          uint32_t h[4], l[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const f2 x = f2_mul(f2_pack(v[2 * e], v[2 * e + 1]), f2_both(wt));
            h[e] = pack_f2(x);
            const f2 hf = f2_pack(__uint_as_float(h[e] << 16), __uint_as_float(h[e] & 0xffff0000u));
            l[e] = pack_f2(f2_fma(hf, f2_both(-1.f), x));
          }
          st_sw128_chunk(hi, row, ch0 + i, make_uint4(h[0], h[1], h[2], h[3]));
          st_sw128_chunk(lo, row, ch0 + i, make_uint4(l[0], l[1], l[2], l[3]));
        }
      }
      fence_proxy_async_smem();
      arrive(S.b_bs[buf]);
    }
  } else if (warp < 24) {
    // ================================================================ output
    const int gt = tid - 512, w = warp & 3, half = (warp - 16) >> 2;
    const int tok0 = 32 * half + 2 * (lane & 3);  // this thread's tokens: tok0 + 8 b and the next, b of 0 .. 3
    // matrix m of a transposed store of four: channels 8 (m & 1), tokens 8 (m >> 1) of 16 x 16; lane 8 m + r gives the
    // address of token r of it
    const int m = lane >> 3, stok = 32 * half + 8 * (m >> 1) + (lane & 7);
    float f[4][2];
    int fn = 0;  // the rows that f is for
    const bool parts = PARTS && q.out_f32;
#pragma unroll 1
    for (int c = 0; c < (states ? 0 : nch); ++c) {
      const int buf = c & 1;
      const int n = chunk_rows(c);
      if (n != fn) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = tok0 + 8 * b + e;
            f[b][e] = i < n ? S.pw[bw ? n - 1 - i : i + 1] * q.iscale : 0.f;
          }
        fn = n;
      }
      const bool stage = n == C;
      if (gt == 0) {  // the store before this one's buffer has read it
        if (parts) bulk_wait_read<0>();
        else bulk_wait_read<1>();
      }
      named_bar(kBarOut, 256);
      wait(S.b_o, c & 1);
      tc_fence_after();
      const uint32_t o1 = lane_addr + TM_O + 32 * half, o2 = o1 + 64;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x[2][8], y[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          tmem_ld_16x256b_x2(o1 + ((16u * h) << 16) + 16 * i, x[i]);
          tmem_ld_16x256b_x2(o2 + ((16u * h) << 16) + 16 * i, y[i]);
        }
        tmem_ld_wait();
        if (h == 1) {
          tc_fence_before();
          arrive(S.b_ofree);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float *fe = f[2 * i + (e >> 2)];
            const f2 xx = f2_pack(x[i][e], x[i][e + 1]), yy = f2_pack(y[i][e], y[i][e + 1]);
            f2_split(f2_fma(yy, f2_pack(fe[0], fe[1]), xx), x[i][e], x[i][e + 1]);
          }
        if (w >= 2 * kc) continue;
        // channels of this thread: d0 and d0 + 8
        const int d0 = 32 * w + 16 * h + (lane >> 2);
        if (stage && parts) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int tok = tok0 + 16 * i + 8 * (e >> 2) + (e & 1), d = d0 + ((e >> 1) & 1) * 8;
              uint8_t *at = sY + w * SZ_PANEL + sw128_chunk_off(tok, (d >> 2) & 7) + (d & 3) * 4;
              *reinterpret_cast<float *>(at) = x[i][e];
            }
        } else if (stage) {
          const int chunk = (32 * w + 16 * h + 8 * (m & 1)) >> 3;
          const uint32_t at = smem_u32(sY + buf * SZ_TILE + (chunk >> 3) * SZ_PANEL) + sw128_chunk_off(stok, chunk & 7);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            stmatrix_x4_trans(at + i * 2048, gdr::pack_bf16(x[i][0], x[i][1]), gdr::pack_bf16(x[i][2], x[i][3]),
                              gdr::pack_bf16(x[i][4], x[i][5]), gdr::pack_bf16(x[i][6], x[i][7]));
        } else {
          const int64_t t0 = chunk_start(c);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int tok = tok0 + 16 * i + 8 * (e >> 2) + (e & 1), d = d0 + ((e >> 1) & 1) * 8;
              if (tok < n && d < Dc) {
                const int64_t at = ((t0 + tok) * p.HV + hv) * Dc + d;
                if (parts) static_cast<float *>(q.out)[at] = x[i][e];
                else static_cast<__nv_bfloat16 *>(q.out)[at] = __float2bfloat16_rn(x[i][e]);
              }
            }
        }
      }
      if (stage) fence_proxy_async_smem();
      named_bar(kBarOut, 256);
      if (gt == 0) {
        if (stage) {
          const int wide = parts ? 32 : 64;  // channels of a panel
          for (int i = 0; i < kc * 64 / wide; ++i)
            tma_store_3d(&maps.y[pi], smem_u32(sY + (parts ? 0 : buf * SZ_TILE) + i * SZ_PANEL), wide * i, (int)hv,
                         (int)chunk_start(c));
        }
        bulk_commit();  // one group a chunk, where nothing is staged an empty one
      }
    }
    if (gt == 0) bulk_wait0();  // every store has landed before the block can exit
  } else if (warp == kProducer && elect_one()) {
    // ================================================================ producer
    const int ha = (int)(hv / q.a.group), hb = (int)(hv / q.b.group), hc = (int)(hv / q.c.group);
    const uint32_t bytes = SZ_PANEL * ((states ? 0 : ka) + ka + kc);
    int issued = 0;
    for (int c = 0; c < nch; ++c) {
      const int st = c % kStages;
      if (c >= kStages) wait(S.empty[st], (c / kStages - 1) & 1);
      if (*err) break;
      const int t0 = (int)chunk_start(c);
      const uint32_t tile = smem_u32(sm + st * SZ_STAGE), bar = smem_u32(&S.full[st]);
      mbar_arrive_expect_tx(bar, bytes);
      for (int i = 0; i < ka; ++i) {
        if (!states) tma_load_3d(tile + i * SZ_PANEL, &maps.a[pi], 64 * i, ha, t0, bar);
        tma_load_3d(tile + SZ_TILE + i * SZ_PANEL, &maps.b[pi], 64 * i, hb, t0, bar);
      }
      for (int i = 0; i < kc; ++i) tma_load_3d(tile + 2 * SZ_TILE + i * SZ_PANEL, &maps.c[pi], 64 * i, hc, t0, bar);
      issued = c + 1;
    }
    // let every copy issued land before the block can exit
    for (int c = issued > kStages ? issued - kStages : 0; c < issued; ++c)
      mbar_wait_drain(smem_u32(&S.full[c % kStages]), (c / kStages) & 1, kTimeout);
  } else if (warp >= kScoreMma && elect_one()) {
    // ================================================================ MMA issuers
    constexpr uint32_t id_sc = idesc_bf16(64, 64, 0, 0), id_o1 = idesc_bf16(128, 64, 1, 0),
                       id_o2 = idesc_bf16(128, 64, 0, 0);
    const uint32_t id_s = idesc_bf16(128, 64 * ka, 1, 1);
    // an operand at base + off has the base's descriptor plus off / 16 in its address field
    auto at = [](uint64_t base, uint32_t off) { return base + (uint64_t)(off >> 4); };
    const uint32_t t0 = smem_u32(sm);
    const uint64_t dk = smem_desc(t0, 16, 1024), dmn = smem_desc(t0, SZ_PANEL, 1024);
    const int last = states && warp != kStateMma ? 0 : nch;
#pragma unroll 1
    for (int c = 0; c < last; ++c) {
      const int st = c % kStages, buf = c & 1;
      const uint32_t ph = (c >> 1) & 1, off = st * SZ_STAGE;
      spin(S.full[st], (c / kStages) & 1);
      if (warp == kScoreMma) {
        if (c > 0) spin(S.b_scfree, (c - 1) & 1);
        if (*err) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t k = off + (ks >> 2) * SZ_PANEL + (ks & 3) * 32;
          if (ks < 4 * ka) mma_bf16(tbase + TM_SC, at(dk, k), at(dk, k + SZ_TILE), id_sc, ks > 0);
        }
        mma_commit(smem_u32(&S.b_sc));
      } else if (warp == kStateMma) {
        spin(S.b_bs[buf], ph);
        if (c > 0) spin(S.b_ufree, (c - 1) & 1);
        if (*err) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint64_t a = at(dmn, off + 2 * SZ_TILE + ks * 2048);
          mma_bf16(tbase + TM_U, a, at(dmn, off + SZ_TILE + ks * 2048), id_s, ks > 0);
          mma_bf16(tbase + TM_U, a, at(dmn, OFF_LO + buf * SZ_TILE + ks * 2048), id_s, 1);
        }
        mma_commit(smem_u32(&S.b_u));
        mma_commit(smem_u32(&S.empty[st]));
      } else {
        spin(S.b_p[buf], ph);
        if (c > 0) spin(S.b_ofree, (c - 1) & 1);
        if (*err) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_bf16(tbase + TM_O, at(dmn, off + 2 * SZ_TILE + ks * 2048), at(dk, OFF_P + buf * SZ_PANEL + ks * 32),
                   id_o1, ks > 0);
        spin(S.b_sb, c & 1);
        if (*err) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          if (ks < 4 * ka)
            mma_bf16_ta(tbase + TM_O + 64, tbase + TM_SB + 8 * ks,
                        at(dk, off + (ks >> 2) * SZ_PANEL + (ks & 3) * 32), id_o2, ks > 0);
        mma_commit(smem_u32(&S.b_o));
        mma_commit(smem_u32(&S.empty[st]));
      }
    }
    // wait for every MMA issued so far before the tensor memory is released
    uint64_t *done = &S.b_final[warp - kScoreMma];
    mma_commit(smem_u32(done));
    mbar_wait_drain(smem_u32(done), 0, kTimeout);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tbase, TM_COLS);
  if (tid == 0 && S.err) raise_status(p.status, GDR_ERR_TIMEOUT);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// [tokens, heads, D] with tokens ld apart, in boxes of 128 bytes of one head's channels and 64 tokens;
// channels from D on read as zeros and are not written.
int make_map(CUtensorMap *m, const LaRows &r, int64_t heads, int64_t tokens, bool f32 = false) {
  const auto fn = encode_fn();
  if (!fn) return set_error(GDR_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[3] = {(cuuint64_t)r.D, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t el = f32 ? 4 : 2, strides[2] = {(cuuint64_t)r.D * el, (cuuint64_t)r.ld * el};
  const cuuint32_t box[3] = {f32 ? 32u : 64u, 1, 64}, es[3] = {1, 1, 1};
  const CUtensorMapDataType type = f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUresult e = fn(m, type, 3, const_cast<void *>(r.p), dims, strides, box, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return e == CUDA_SUCCESS ? GDR_OK : set_error(GDR_ERR_CUDA, "cuTensorMapEncodeTiled failed");
}

// What TMA can describe: 16-byte aligned bases, rows and heads.
bool tma_ok(const LaRows &r) { return r.D <= 128 && r.D % 8 == 0 && r.ld % 8 == 0 && is_aligned16(r.p); }

}  // namespace

bool tc_takes(const LaArgs &p, int passes, int dtype) {
  if (dtype != GDR_BF16 || p.tokens == 0 || p.N == 0) return false;
  for (int i = 0; i < passes; ++i) {
    const LaPass &q = p.pass[i];
    if (!tma_ok(q.a) || !tma_ok(q.b) || !tma_ok(q.c) || !is_aligned16(q.out)) return false;
  }
  return true;
}

int launch_tc(const LaArgs &p, int passes, cudaStream_t st) {
  Maps maps{};
  for (int i = 0; i < passes; ++i) {
    const LaPass &q = p.pass[i];
    const LaRows y{q.out, p.HV * q.c.D, q.c.D, 1};
    const auto map = [&](CUtensorMap *m, const LaRows &r) { return make_map(m, r, p.HV / r.group, p.tokens); };
    int rc;
    if ((rc = map(&maps.b[i], q.b)) != GDR_OK || (rc = map(&maps.c[i], q.c)) != GDR_OK) return rc;
    if (p.mode == kStates) continue;
    if ((rc = map(&maps.a[i], q.a)) != GDR_OK) return rc;
    if ((rc = make_map(&maps.y[i], y, p.HV, p.tokens, q.out_f32)) != GDR_OK) return rc;
  }
  const int64_t items = std::max<int64_t>(1, (p.mode == kWhole ? p.N : p.slots) * p.HV);
  if (items * passes > 0x7fffffff) return set_error(GDR_ERR_SHAPE, "too many sequences and heads for one launch");
  bool parts = false;
  for (int i = 0; i < passes; ++i) parts |= p.mode != kStates && p.pass[i].out_f32;
  bool wide = false;
  for (int i = 0; i < passes; ++i) wide |= p.pass[i].a.D > 64 || p.pass[i].c.D > 64;
  const auto kernel = wide ? parts ? la_tc_kernel<true, 2> : la_tc_kernel<false, 2>
                           : parts ? la_tc_kernel<true, 1> : la_tc_kernel<false, 1>;
  const int smem = (int)(wide ? smem_bytes<2>() : smem_bytes<1>());
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute(la_tc_kernel)");
  kernel<<<(unsigned)(items * passes), kTcThreads, smem, st>>>(maps, p, passes);
  return launched("la_tc_kernel");
}

}  // namespace la
}  // namespace gdr
